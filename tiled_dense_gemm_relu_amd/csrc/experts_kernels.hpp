// An expert layer for a few tokens (gemm_relu_blocks.h) in two launches: routing
// and the first products, then the second products and their sum.
//
// With a few tokens the time is that of reading the chosen experts' weights, once.
// Every workgroup makes the routing table for itself (tokens are few), so nothing
// waits for it, and takes units of 16 of an expert's rows (an expert with more has
// several) and 16 NB output columns; its waves take pieces of k in turn and add their
// sums in LDS.  The rows stream with the weights through a ring of each wave's own in
// LDS, by DMA, as in blocks_stream.hpp; operands whose rows DMA cannot read (odd
// lengths, 2-byte alignment) go through registers.
//
// The first launch leaves weight * ReLU(sum) of every choice as a sum of two 16-bit
// values, for the second one's matrix instructions: off by at most 2^-16 of the value or
// 2^-134 with bf16, with fp16 by 2^-22 or 2^-25, and infinite past 65504 (one value would be off
// by 2^-9 and 2^-12; a third takes half as much again of the rings' room for rows).
// The second launch's units write a choice's products as fp32; the last unit of a column
// block to end adds each token's in the order of its choices.
//
// 24 tokens, 4 of 64 experts, 8-bit 2048 x 4096: 139 us, 6 TB/s of the chosen experts'
// weights.  One token, 4 experts, 16-bit 2048 x 2048: two launches of 12.5 us, each a
// chain of launch, table, first bytes and 33 MB.
#pragma once

#include <type_traits>

#include "blocks_bytes.hpp"
#include "blocks_table.hpp"
#include "groups_skinny.hpp"

namespace gemm_relu_hip {

// Who goes where: slot t top + j is token t's choice j.  In dynamic LDS, as large as
// the call needs (route_table_bytes).
struct RouteTable {
    int16_t* ids;            // a slot's expert, -1: none
    float* weights;          // a slot's weight
    int* count;              // an expert's slots
    uint32_t* tiles;         // row tiles of the experts that have slots: expert, and first row << 16
    int* n_tiles;
    uint16_t* sorted;        // slots by expert, in order
    uint16_t* end;           // where an expert's slots end in `sorted`

    __device__ __forceinline__ RouteTable(uint8_t* p, int slots, int experts)
    {
        ids = reinterpret_cast<int16_t*>(p);
        weights = reinterpret_cast<float*>(ids + (slots + 1) / 2 * 2);
        count = reinterpret_cast<int*>(weights + slots);
        tiles = reinterpret_cast<uint32_t*>(count + experts);
        n_tiles = reinterpret_cast<int*>(tiles + min(experts, slots) + slots / 16);
        sorted = reinterpret_cast<uint16_t*>(n_tiles + 1);
        end = sorted + slots;
    }
};

__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    const int m = wave_scan((int)v, [](int a, int b) { return (int)max((uint32_t)a, (uint32_t)b); });
    return (uint32_t)__builtin_amdgcn_readlane(m, 63);
}

__device__ __forceinline__ float wave_sum(float v)
{
    const int s = wave_scan(__builtin_bit_cast(int, v), [](int a, int b) {
        return __builtin_bit_cast(int, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
    });
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(s, 63));
}

// The choices of N tokens by one wave: of each token the largest logits, ties to the
// lowest index, and their softmax weights; lane j gets choice j.  l[n][r] is logit
// 64 r + lane of token n (-inf past the last).  The tokens' steps are independent, so
// their chains of moves between lanes overlap.  Logits are compared as unsigned keys in
// their order; key 0 is never chosen (-inf, and what has been chosen).
template <int N, int R>
__device__ __forceinline__ void choose(float (&l)[N][R], int top, bool renormalize, int lane, int (&id)[N], float (&weight)[N])
{
    uint32_t key[N][R];
    bool bad[N];
    float largest[N], mine[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        bad[n] = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            l[n][r] += 0.0f;                              // (-0 and +0 are equal)
            const uint32_t bits = __builtin_bit_cast(uint32_t, l[n][r]);
            bad[n] |= !(l[n][r] < __builtin_inff());
            key[n][r] = l[n][r] == -__builtin_inff() ? 0u : (bits & 0x80000000u) ? ~bits : bits | 0x80000000u;
        }
        bad[n] = __ballot(bad[n]) != 0;
        id[n] = -1;
        largest[n] = mine[n] = 0.0f;
    }
    for (int j = 0; j < top; ++j) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            uint32_t m = 0;
#pragma unroll
            for (int r = 0; r < R; ++r) m = max(m, key[n][r]);
            m = wave_max(m);
            bool found = m == 0 || bad[n];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint64_t at = __ballot(key[n][r] == m);
                if (found || !at) continue;
                found = true;
                const int who = __builtin_ctzll(at);
                const float value = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, l[n][r]), who));
                if (j == 0) largest[n] = value;
                if (lane == who) key[n][r] = 0;
                if (lane == j) {
                    id[n] = 64 * r + who;
                    mine[n] = value;
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const float e = id[n] >= 0 ? expf(mine[n] - largest[n]) : 0.0f;
        float sum = 0.0f;
        if (renormalize) {
            sum = e;
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) sum += l[n][r] == -__builtin_inff() ? 0.0f : expf(l[n][r] - largest[n]);
        }
        sum = wave_sum(sum);
        weight[n] = bad[n] ? __builtin_nanf("") : id[n] >= 0 ? e / sum : 0.0f;
    }
}

// Tokens first, first + stride, ..., of `tokens`, by one wave.
template <int N, int R, class Put>
__device__ __forceinline__ void route(const float* __restrict__ logits, int tokens, int experts, int top, bool renormalize, int first,
                                      int stride, int lane, Put put)
{
    for (int token = first; token < tokens; token += N * stride) {
        float l[N][R];
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int r = 0; r < R; ++r)
                l[n][r] = 64 * r + lane < experts && token + n * stride < tokens
                              ? logits[(size_t)(token + n * stride) * (size_t)experts + (size_t)(64 * r + lane)] : -__builtin_inff();
        int id[N];
        float weight[N];
        choose<N, R>(l, top, renormalize, lane, id, weight);
        if (lane < top) {
#pragma unroll
            for (int n = 0; n < N; ++n)
                if (token + n * stride < tokens) put((token + n * stride) * top + lane, id[n], weight[n]);
        }
    }
}

template <class Put>
__device__ __forceinline__ void route_any(const float* logits, int tokens, int experts, int top, bool renormalize, int first, int stride,
                                          int lane, Put put)
{
    if (experts <= 64) route<4, 1>(logits, tokens, experts, top, renormalize, first, stride, lane, put);
    else if (experts <= 256) route<1, 4>(logits, tokens, experts, top, renormalize, first, stride, lane, put);
    else route<1, kMaxExperts / 64>(logits, tokens, experts, top, renormalize, first, stride, lane, put);
}

// Routing by itself, a wave a token: where every workgroup's doing it again would cost more
// than a launch.
static __global__ __launch_bounds__(64) void route_tokens(ExpertsArgs a)
{
    route_any(a.logits, a.tokens, a.experts, a.top, a.renormalize != 0, (int)blockIdx.x, (int)gridDim.x, (int)threadIdx.x,
              [&](int slot, int id, float weight) {
                  a.ids[slot] = id;
                  a.weights[slot] = weight;
              });
}

// The routing table, by the whole workgroup, with row tiles of ROWS rows.  With logits
// the choices are made here and, by the first workgroup, written.
template <int WAVES, int ROWS>
__device__ inline void make_table(const RouteTable& t, const ExpertsArgs& a, int lane, int wave)
{
    constexpr int THREADS = 64 * WAVES;
    const int slots = a.tokens * a.top, tid = threadIdx.x;
    for (int e = tid; e < a.experts; e += THREADS) t.count[e] = 0;
    if (a.logits) {
        route_any(a.logits, a.tokens, a.experts, a.top, a.renormalize != 0, wave, WAVES, lane, [&](int slot, int id, float weight) {
            t.ids[slot] = (int16_t)id;
            t.weights[slot] = weight;
            if (blockIdx.x == 0) {
                a.ids[slot] = id;
                a.weights[slot] = weight;
            }
        });
    } else {
        for (int s = tid; s < slots; s += THREADS) {
            const int id = a.ids[s];
            t.ids[s] = (int16_t)(id >= 0 && id < a.experts ? id : -1);
            t.weights[s] = a.weights[s];
        }
    }
    __syncthreads();
    for (int s = tid; s < slots; s += THREADS)
        if (t.ids[s] >= 0) atomicAdd(&t.count[t.ids[s]], 1);
    __syncthreads();
    if (wave == 0) {
        int before = 0, tiles = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 64) {
            const int c = e0 + lane < a.experts ? t.count[e0 + lane] : 0, incl = wave_scan_sum(c);
            const int n = (c + ROWS - 1) / ROWS, at = wave_scan_sum(n);
            if (c > 0) {
                t.end[e0 + lane] = (uint16_t)(before + incl - c);
                for (int i = 0; i < n; ++i) t.tiles[tiles + at - n + i] = (uint32_t)(e0 + lane) | ((uint32_t)(i * ROWS) << 16);
            }
            before += __builtin_amdgcn_readlane(incl, 63);
            tiles += __builtin_amdgcn_readlane(at, 63);
        }
        if (lane == 0) *t.n_tiles = tiles;
        // The slots in order, 64 at a time: those of one expert find each other by the bits of
        // its number, and `end`, where they begin at first, moves on past them.
        const int bits = 32 - __builtin_clz(a.experts);
        for (int s0 = 0; s0 < slots; s0 += 64) {
            const int s = s0 + lane, id = s < slots ? t.ids[s] : -1;
            uint64_t same = __ballot(id >= 0);
            for (int b = 0; b < bits; ++b) {
                const uint64_t set = __ballot((id >> b) & 1);
                same &= (id >> b) & 1 ? set : ~set;
            }
            if (id >= 0) {
                const int at = t.end[id], rank = __popcll(same & ((uint64_t(1) << lane) - 1)), n = __popcll(same);
                t.sorted[at + rank] = (uint16_t)s;
                if (rank == n - 1) t.end[id] = (uint16_t)(at + n);
            }
            __builtin_amdgcn_wave_barrier();
        }
    }
    __syncthreads();
}

// The scale of a block of 8-bit weights as two factors: a power of two that the widened
// weights take, and the rest, which their sum does.  bf16 rows times stored values could
// pass the largest float where the products do not: weights with small scales take as much
// of them as keeps 128 products of any rows below it.  (Small rows need nothing: the
// products of 8 and 4 bits are exact, subnormal ones too.  Nor do fp16 rows, whose products
// are at most 2^32.)
struct WeightScale {
    float power, rest;
};
template <int DT, int FORMAT>
__device__ __forceinline__ WeightScale weight_scale(float s)
{
    if constexpr (DT == kF16) return WeightScale{1.0f, s};
    constexpr int least = FORMAT == kE4M3 ? -16 : -23;      // 128 448 2^128 2^-16 < 2^128; 128 57344 2^128 2^-23 < 2^128
    const int e = min(max((int)((__builtin_bit_cast(uint32_t, s) >> 23) & 0xffu) - 127, least), 0);
    return WeightScale{__builtin_bit_cast(float, (uint32_t)(e + 127) << 23), __builtin_ldexpf(s, -e)};
}

// 8 weights of a lane from 8 bytes, times a power of two, as 16-bit values (exact).
template <int DT, int FORMAT>
__device__ __forceinline__ u32x4 widen(uint32_t lo, uint32_t hi, float power)
{
    u32x4 r;
#define GEMM_RELU_WIDEN(NAME) \
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_##NAME(lo, power, false)); \
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_##NAME(lo, power, true)); \
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_##NAME(hi, power, false)); \
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_##NAME(hi, power, true));
    if constexpr (DT == kF16 && FORMAT == kE4M3) {
        GEMM_RELU_WIDEN(f16_fp8)
    } else if constexpr (DT == kF16) {
        GEMM_RELU_WIDEN(f16_bf8)
    } else if constexpr (FORMAT == kE4M3) {
        GEMM_RELU_WIDEN(bf16_fp8)
    } else {
        GEMM_RELU_WIDEN(bf16_bf8)
    }
#undef GEMM_RELU_WIDEN
    return r;
}

// Storage of the weights: 16-bit (out, in) or (in, out) in X's dtype, or 8-bit (out, in).
enum { kStoreNK = 0, kStoreKN = 1, kStoreE4M3 = 2, kStoreE5M2 = 3 };

typedef uint32_t u32x3 __attribute__((ext_vector_type(3)));

// A lane's weights of a piece, on their way: 16 columns x 128 k in NB blocks.
//  NK: [block][k-step] 8 consecutive k of column 16 block + lane % 16.
//  KN: [k-step][k] 4 consecutive columns 4 (lane % 16) .. of k-step's k 8 kb .., in 3
//      dwords, which hold them at 2-byte alignment too.
//  8-bit: [block][half] 16 consecutive k.
template <int STORE, bool ODD, int NB>
struct PieceWeights;
template <bool ODD, int NB>
struct PieceWeights<kStoreNK, ODD, NB> {
    SkinnyChunk<ODD> v[NB][4];
};
template <bool ODD, int NB>
struct PieceWeights<kStoreKN, ODD, NB> {
    static_assert(NB == 4, "4 columns a lane");
    u32x3 v[4][8];
};
template <bool ODD, int NB>
struct PieceWeights<kStoreE4M3, ODD, NB> {
    u32x4 v[NB][2];
};
template <bool ODD, int NB>
struct PieceWeights<kStoreE5M2, ODD, NB> : PieceWeights<kStoreE4M3, ODD, NB> {};

// The sums over pieces p0 + wave, p0 + wave + WAVES, .. of a unit's NB blocks of columns.
//  Rows: lane's row is x_off bytes into rx (kOobOffset: none); with SPLIT_X also its low
//  parts, x_low bytes on.
template <int DT, int STORE, bool SPLIT_X, int NB, int WAVES>
__device__ __forceinline__ void expert_sums(floatx4 (&acc)[NB], const AnyRsrc& rx, uint32_t x_off, uint32_t x_low,
                                            const uint8_t* w, const float* scales, int64_t ld, int n0, int in, int out,
                                            int p0, int p1, int wave, int lane)
{
    constexpr bool WIDE = STORE >= kStoreE4M3, ODD = !WIDE, ODD_X = !SPLIT_X;
    constexpr int FORMAT = STORE == kStoreE4M3 ? kE4M3 : kE5M2;
    constexpr int KU = NB <= 2 ? 2 : 1;                // pieces in flight
    const int r16 = lane & 15, g = lane >> 4;
    const int cols = min(16 * NB, out - n0);
    // NK and 8-bit: rows n0 .. of the expert's weights
    AnyRsrc rw{};
    if constexpr (STORE == kStoreNK) rw = make_any_rsrc(reinterpret_cast<const uint16_t*>(w + (size_t)n0 * (size_t)ld), (uint32_t)cols * (uint32_t)ld);
    if constexpr (WIDE) rw.rsrc = make_rsrc(w + (size_t)n0 * (size_t)ld, (uint32_t)cols * (uint32_t)ld);
    // 8 k of step s of piece p: 8-bit weights have 16 consecutive ones a lane.
    auto first_k = [&](int p, int s) { return p * kBlock + (WIDE ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g); };
    auto load_x = [&](int p, int s, SkinnyChunk<ODD_X>& high, SkinnyChunk<ODD_X>& low) {
        const int k = first_k(p, s);
        const uint32_t off = p < p1 && x_off != kOobOffset && k < in ? x_off + (uint32_t)k * 2u : kOobOffset;
        high = load_skinny<ODD_X>(rx, off);
        if constexpr (SPLIT_X) low = load_skinny<ODD_X>(rx, off == kOobOffset ? kOobOffset : off + x_low);
    };
    for (int i0 = p0 + wave; i0 < p1; i0 += KU * WAVES) {
        PieceWeights<STORE, ODD, NB> pw[KU];
        // A piece's rows of X are in flight with its weights.
        SkinnyChunk<ODD_X> x[KU][4], low[SPLIT_X ? KU : 1][4];
        float scale[KU];
#pragma unroll
        for (int q = 0; q < KU; ++q) {
            const int p = i0 + q * WAVES, k0 = p * kBlock;
            const bool live = p < p1;
            if constexpr (STORE == kStoreNK) {
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        pw[q].v[i][s] = load_skinny<ODD>(rw, live ? (uint32_t)(16 * i + r16) * (uint32_t)ld + (uint32_t)(k0 + 32 * s + 8 * g) * 2u : kOobOffset);
            } else if constexpr (STORE == kStoreKN) {
                const int k1 = live ? min(k0, in) : 0;
                const AnyRsrc rp = make_any_rsrc(reinterpret_cast<const uint16_t*>(w) + (size_t)k1 * (size_t)out + n0,
                                                 live ? (uint32_t)(max(0, min(kBlock, in - k1)) * (int64_t)out - n0) * 2u : 0u);
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t off = 4 * r16 < cols ? ((uint32_t)(32 * s + 8 * g + e) * (uint32_t)out + 4u * (uint32_t)r16) * 2u : kOobOffset;
                        pw[q].v[s][e] = __builtin_amdgcn_raw_buffer_load_b96(rp.rsrc, (off + rp.shift) & ~3u, 0, 0);
                    }
            } else {
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int k = k0 + 64 * h + 16 * g;
                        pw[q].v[i][h] = __builtin_amdgcn_raw_buffer_load_b128(rw.rsrc, live && k < in ? (uint32_t)(16 * i + r16) * (uint32_t)ld + (uint32_t)k : kOobOffset, 0, 0);
                    }
                scale[q] = live ? scales[p] : 0.0f;
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) load_x(p, s, x[q][s], low[SPLIT_X ? q : 0][s]);
        }
#pragma unroll
        for (int q = 0; q < KU; ++q) {
            const int p = i0 + q * WAVES, k0 = p * kBlock;
            if (p >= p1) break;
            const bool tail = k0 + kBlock > in;
            floatx4 sum[WIDE ? NB : 1];
            WeightScale block_scale{1.0f, 1.0f};
            if constexpr (WIDE) {
                block_scale = weight_scale<DT, FORMAT>(scale[q]);
#pragma unroll
                for (int i = 0; i < NB; ++i) sum[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int k = first_k(p, s), valid = in - k;
                u32x4 wv[NB];
                if constexpr (STORE == kStoreNK) {
#pragma unroll
                    for (int i = 0; i < NB; ++i) {
                        wv[i] = skinny_value<ODD>(pw[q].v[i][s], rw, (uint32_t)(16 * i + r16) * (uint32_t)ld + (uint32_t)k * 2u);
                        if (tail) wv[i] = keep_first(wv[i], valid);
                    }
                } else if constexpr (STORE == kStoreKN) {
                    // [k] x 4 columns -> [column] x 8 k
                    const uint32_t base = (uint32_t)((uintptr_t)(reinterpret_cast<const uint16_t*>(w) + (size_t)k0 * (size_t)out + n0)) & 2u;
                    u32x2 row[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const u32x3 v = pw[q].v[s][e];
                        const uint32_t bits = ((uint32_t)(e & 1) * (uint32_t)out * 2u + base & 2u) * 8u;      // (even rows are alike)
                        row[e] = u32x2{__builtin_amdgcn_alignbit(v.y, v.x, bits), __builtin_amdgcn_alignbit(v.z, v.y, bits)};
                        if (tail && e >= valid) row[e] = u32x2{0u, 0u};
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int h = 0; h < 4; ++h)
                            wv[c][h] = __builtin_amdgcn_perm(row[2 * h + 1][c >> 1], row[2 * h][c >> 1], (c & 1) ? 0x07060302u : 0x05040100u);
                } else {
#pragma unroll
                    for (int i = 0; i < NB; ++i) {
                        u32x2 b{pw[q].v[i][s >> 1][2 * (s & 1)], pw[q].v[i][s >> 1][2 * (s & 1) + 1]};
                        if (tail) {
                            const u32x4 kept = keep_bytes(u32x4{b.x, b.y, 0u, 0u}, valid);
                            b = u32x2{kept[0], kept[1]};
                        }
                        wv[i] = widen<DT, FORMAT>(b.x, b.y, block_scale.power);
                    }
                }
                u32x4 xv = skinny_value<ODD_X>(x[q][s], rx, x_off + (uint32_t)k * 2u);
                if (tail) xv = keep_first(xv, valid);
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    floatx4& to = WIDE ? sum[WIDE ? i : 0] : acc[i];
                    to = mfma_16x16x32<DT>(wv[i], xv, to);
                }
                if constexpr (SPLIT_X) {
                    u32x4 lv = low[q][s].v;
                    if (tail) lv = keep_first(lv, valid);
#pragma unroll
                    for (int i = 0; i < NB; ++i) {
                        floatx4& to = WIDE ? sum[WIDE ? i : 0] : acc[i];
                        to = mfma_16x16x32<DT>(wv[i], lv, to);
                    }
                }
            }
            if constexpr (WIDE) {
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][e] = __builtin_fmaf(block_scale.rest, sum[i][e], acc[i][e]);
            }
        }
    }
}

// The sums over this wave's pieces (64 k of 16-bit weights, 128 of 8-bit ones: 128
// bytes of a row of W, or 64 rows of 64 columns) for up to 16 rows, through its ring
// of S stages: W, then X's rows in halves of 64 k, then their low parts.
//  x_row[q]: where the row of X of this lane's 16 bytes of DMA instruction q begins,
// in bytes (kOobOffset: none).
// ONCE: W does not stay in the caches.
template <int DT, int STORE, bool SPLIT_X, bool ONCE, int NB, int S, int WAVES>
__device__ __forceinline__ void expert_stream(floatx4 (&acc)[NB], const uint16_t* x, uint32_t x_bytes, const uint32_t (&x_row)[2],
                                              uint32_t x_low, const uint8_t* w, const float* scales, int64_t ld, int n0, int in,
                                              int out, int p0, int p1, uint8_t* ring, int turn, int wave, int lane)
{
    constexpr bool WIDE = STORE >= kStoreE4M3, KN = STORE == kStoreKN;
    constexpr int FORMAT = STORE == kStoreE4M3 ? kE4M3 : kE5M2;
    constexpr int K = WIDE ? 128 : 64, HALVES = K / 64, W_BYTES = NB * 2048, X_BYTES = 2048;
    constexpr int STAGE = W_BYTES + HALVES * X_BYTES * (SPLIT_X ? 2 : 1), NQ = STAGE / 1024;
    static_assert(!KN || NB == 4, "rows of 128 bytes");
    const int r16 = lane & 15, g = lane >> 4, kb = kgroup16(g);
    const int count = p1 - p0, mine = count > wave ? (count - wave + WAVES - 1) / WAVES : 0;
    const int cols = min(16 * NB, out - n0);
    const uint32_t ring_lds = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) uint8_t*)ring);
    auto piece_at = [&](int i) {
        const int p = wave + i * WAVES;
        return p0 + (p + turn < count ? p + turn : p + turn - count);
    };
    // A lane's 16 bytes of an instruction of 8 rows; k-contiguous rows are swizzled by
    // a_swizzle (period 16 rows), (K, N) rows by b_swizzle (32 rows, two of them alike).
    uint32_t w_off[2];
    int pos[2];                   // first byte of the lane's piece in its 128
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int row = 8 * q + lane / 8;
        pos[q] = ((lane % 8) ^ a_swizzle<128>(row)) * 16;
        if constexpr (KN) {
            const int k = 16 * q + lane / 8, c = ((lane % 8) ^ b_swizzle<128, 16>(k)) * 16;   // (k and k + 8 are alike)
            w_off[q] = c < 2 * cols ? (uint32_t)(lane / 8) * (uint32_t)ld + (uint32_t)c : kOobOffset;
        } else {
            w_off[q] = (uint32_t)row * (uint32_t)ld + (uint32_t)pos[q];
        }
    }
    auto uniform = [](const void* p, uint32_t bytes) {
        const int32x4_t r = rsrc_words(p, bytes);
        return int32x4_t{__builtin_amdgcn_readfirstlane(r[0]), __builtin_amdgcn_readfirstlane(r[1]),
                         __builtin_amdgcn_readfirstlane(r[2]), kBufferFlags};
    };
    float scale[S];
    const int32x4_t rx = uniform(x, x_bytes);
    auto fill = [&](int i, int slot, float& s) __attribute__((always_inline)) {
        const bool live = i < mine;
        const int p = __builtin_amdgcn_readfirstlane(piece_at(live ? i : 0)), k0 = p * K, left = live ? in - k0 : 0;   // elements
        const uint32_t to = (uint32_t)__builtin_amdgcn_readfirstlane((int)(ring_lds + (uint32_t)(slot * STAGE)));
        const auto weights = [&](auto&& load) __attribute__((always_inline)) {
            if constexpr (KN) {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int k = k0 + 8 * q;
                    // up to the end of the last row
                    const uint32_t bytes = left > 8 * q ? (uint32_t)min(8, left - 8 * q) * (uint32_t)ld - 2u * (uint32_t)n0 : 0u;
                    load(uniform(w + (size_t)min(k, in) * (size_t)ld + 2 * (size_t)n0, bytes), to + q * 1024, w_off[(q >> 1) & 1], 0u);
                }
            } else {
#pragma unroll
                for (int q = 0; q < 2 * NB; ++q) {
                    const int skip = 16 * (q >> 1);
                    load(uniform(w + (size_t)(n0 + skip) * (size_t)ld, (uint32_t)max(0, cols - skip) * (uint32_t)ld), to + q * 1024,
                         pos[q & 1] < (WIDE ? left : 2 * left) ? w_off[q & 1] : kOobOffset, (uint32_t)(WIDE ? k0 : 2 * k0));
                }
            }
        };
        if constexpr (ONCE) weights(dma_b128_once);
        else weights(dma_b128);
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const uint32_t off = x_row[q] != kOobOffset && 128 * h + pos[q] < 2 * left ? x_row[q] + (uint32_t)pos[q] : kOobOffset;
                const uint32_t at = to + W_BYTES + (2 * h + q) * 1024, soff = (uint32_t)(2 * k0 + 128 * h);
                dma_b128(rx, at, off, soff);
                if constexpr (SPLIT_X) dma_b128(rx, at + HALVES * X_BYTES, off, soff + x_low);
            }
        if constexpr (WIDE) s = live ? scales[p] : 0.0f;
    };
#pragma unroll
    for (int s = 0; s < S; ++s) fill(s, s, scale[s]);
    for (int i0 = 0; i0 < mine; i0 += S) {
#pragma unroll
        for (int slot = 0; slot < S; ++slot) {
            const int i = i0 + slot;
            if (i >= mine) break;
            wait_vmcnt<(S - 1) * NQ>();
            WeightScale block_scale{1.0f, 1.0f};
            if constexpr (WIDE) {
                // (taken from its load here: a wait for it behind the next fill would wait for that too)
                block_scale = weight_scale<DT, FORMAT>(scale[slot]);
                asm volatile("" : "+v"(block_scale.power), "+v"(block_scale.rest));
            }
            const uint8_t *const st = ring + slot * STAGE, *const sx = st + W_BYTES;
            constexpr int STEPS = WIDE ? 4 : 2;                  // of 32 k
            u32x4 wf[NB][2], xf[STEPS], lf[SPLIT_X ? STEPS : 1];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (KN) {
                        const int krow = 8 * kb + (r16 >> 2), n = 16 * b + 4 * (r16 & 3);
                        const uint8_t* q = st + (krow + 32 * h) * 128 + 16 * ((n >> 3) ^ b_swizzle<128, 16>(krow)) + 8 * (r16 & 1);
                        const u32x2 lo = ds_read_tr16(q), hi = ds_read_tr16(q + 4 * 128);
                        wf[b][h] = u32x4{lo.x, lo.y, hi.x, hi.y};
                    } else {
                        wf[b][h] = *reinterpret_cast<const u32x4*>(st + b * 2048 + r16 * 128 + 16 * ((4 * h + kb) ^ a_swizzle<128>(r16)));
                    }
                }
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                // 8-bit weights have 16 consecutive k a lane
                const int half = WIDE ? s >> 1 : 0, chunk = WIDE ? 2 * kb + (s & 1) : 4 * s + kb;
                const uint8_t* q = sx + half * X_BYTES + r16 * 128 + 16 * (chunk ^ a_swizzle<128>(r16));
                xf[s] = *reinterpret_cast<const u32x4*>(q);
                if constexpr (SPLIT_X) lf[s] = *reinterpret_cast<const u32x4*>(q + HALVES * X_BYTES);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");     // the slot has been read
            fill(i + S, slot, scale[slot]);
            const int k0 = piece_at(i) * K;
            floatx4 sum[WIDE ? NB : 1];
            if constexpr (WIDE) {
#pragma unroll
                for (int b = 0; b < NB; ++b) sum[b] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
            }
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int valid = in - (k0 + (WIDE ? 64 * (s >> 1) + 16 * kb + 8 * (s & 1) : 32 * s + 8 * kb));
                const bool tail = k0 + K > in;
                if (tail) {
                    xf[s] = keep_first(xf[s], valid);
                    if constexpr (SPLIT_X) lf[s] = keep_first(lf[s], valid);
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    u32x4 wv;
                    if constexpr (WIDE) {
                        u32x2 v{wf[b][s >> 1][2 * (s & 1)], wf[b][s >> 1][2 * (s & 1) + 1]};
                        if (tail) {
                            const u32x4 kept = keep_bytes(u32x4{v.x, v.y, 0u, 0u}, valid);
                            v = u32x2{kept[0], kept[1]};
                        }
                        wv = widen<DT, FORMAT>(v.x, v.y, block_scale.power);
                    } else {
                        wv = wf[b][s];
                        if (tail && !KN) wv = keep_first(wv, valid);    // ((K, N) rows past the last are zeros)
                    }
                    floatx4& to = WIDE ? sum[WIDE ? b : 0] : acc[b];
                    if constexpr (SPLIT_X) to = mfma_16x16x32<DT>(wv, lf[s], to);
                    to = mfma_16x16x32<DT>(wv, xf[s], to);
                }
            }
            if constexpr (WIDE) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[b][e] = __builtin_fmaf(block_scale.rest, sum[b][e], acc[b][e]);
            }
        }
    }
    wait_vmcnt<0>();              // nothing lands in the ring after this
}

// KIND: kExpertBlocks columns, kExpertWaves waves.  ODD: everything through registers.
template <int DT, int STORE, bool ODD, bool SECOND, int KIND>
__global__ __launch_bounds__(64 * kExpertWaves[KIND], KIND == 1 ? ODD || STORE >= kStoreE4M3 ? 2 : 3 : 1) void expert_products(ExpertsArgs a)
{
    constexpr bool WIDE = STORE >= kStoreE4M3, KN = STORE == kStoreKN;
    constexpr int kDeviceScope = 16;   // cache policy sc1
    constexpr int NB = KN ? 4 : kExpertBlocks[KIND], WAVES = kExpertWaves[KIND], THREADS = 64 * WAVES;
    constexpr int COLS = 16 * NB, PART = COLS * 17, STAGE = NB * 2048 + (WIDE ? 4096 : 2048) * (SECOND ? 2 : 1);
    constexpr int S = KIND == 0 && STORE == kStoreNK ? 2 : 1;
    constexpr int PARTS = WAVES * PART * 4, RING = ODD ? 0 : WAVES * S * STAGE;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[RING > PARTS ? RING : PARTS];
    __shared__ int before;
    extern __shared__ __attribute__((aligned(16))) uint8_t table[];
    float* const part = reinterpret_cast<float*>(smem);       // the waves' sums, after the rings
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), tid = threadIdx.x;
    const int r16 = lane & 15, g = lane >> 4;
    const RouteTable t(table, a.tokens * a.top, a.experts);
    make_table<WAVES, kExpertRows>(t, a, lane, wave);
    const int blocks_n = (a.out + COLS - 1) / COLS, scale_blocks = (a.in + kBlock - 1) / kBlock;
    const int tiles = __builtin_amdgcn_readfirstlane(*t.n_tiles);
    const int units = tiles * blocks_n * a.splits;
    // Where column c of a unit sits in its rows of LDS: in registers (K, N) weights give a
    // lane 4 neighbouring columns, one in each block.
    auto column = [](int c) { return KN && ODD ? (c & 3) * 16 + (c >> 2) : c; };

    // Rows of tokens without a choice, where no unit would write them; with logits that
    // cannot be ranked the row is NaN.
    auto row_without = [&](int token) {
        return a.routed && t.ids[token * a.top] < 0 && t.weights[token * a.top] != t.weights[token * a.top] ? __builtin_nanf("") : 0.0f;
    };
    if (SECOND && tiles == 0) {
        for (int64_t i = (int64_t)blockIdx.x * THREADS + tid; i < (int64_t)a.tokens * a.out; i += (int64_t)gridDim.x * THREADS)
            a.y[i] = act_cast<DT>(row_without((int)(i / a.out)), false);
        return;
    }
    const uint32_t x_bytes = SECOND ? (uint32_t)(a.tokens * a.top) * (uint32_t)a.mid_row * 4u : (uint32_t)a.tokens * (uint32_t)a.in * 2u;
    const AnyRsrc rx = make_any_rsrc(a.x, x_bytes);
    for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int nb = unit % blocks_n, rest = unit / blocks_n, split = rest % a.splits, n0 = nb * COLS;
        const uint32_t tile = (uint32_t)__builtin_amdgcn_readfirstlane((int)t.tiles[rest / a.splits]);
        const int expert = (int)(tile & 0xffffu), row0 = (int)(tile >> 16);
        const int count = __builtin_amdgcn_readfirstlane(t.count[expert]), first = __builtin_amdgcn_readfirstlane(t.end[expert]) - count;
        const uint8_t* w = a.w + (size_t)expert * (size_t)(KN ? a.in : a.out) * (size_t)a.ld;
        const float* scales = WIDE ? a.scales + ((size_t)expert * (size_t)((a.out + kBlock - 1) / kBlock) + (size_t)(n0 / kBlock)) * (size_t)scale_blocks
                                   : nullptr;
        // where a row of X begins, in bytes
        auto row_of_x = [&](int r) {
            const int slot = t.sorted[first + min(r, count - 1)];
            return r >= count ? kOobOffset : SECOND ? (uint32_t)slot * (uint32_t)a.mid_row * 4u : (uint32_t)(slot / a.top) * (uint32_t)a.in * 2u;
        };
        // The unit's share of `pieces` of k.
        auto from = [&](int pieces, int s) { return (int)((int64_t)pieces * s / a.splits); };
        // Adds the waves' sums and hands them on.
        auto finish = [&](const floatx4 (&sums)[NB]) __attribute__((always_inline)) {
            __syncthreads();           // the rings are read
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) part[wave * PART + (16 * i + 4 * g + e) * 17 + r16] = sums[i][e];
            __syncthreads();
            for (int o = tid; o < 16 * COLS; o += THREADS) {
                const int row = o / COLS, c = o % COLS, r = row0 + row;
                if (r >= count || n0 + c >= a.out) continue;
                float z = 0.0f;
#pragma unroll
                for (int v = 0; v < WAVES; ++v) z += part[v * PART + column(c) * 17 + row];
                const int slot = t.sorted[first + r];
                if constexpr (SECOND) {
                    __hip_atomic_store(a.part + ((size_t)slot * (size_t)a.splits + (size_t)split) * (size_t)a.out + (size_t)(n0 + c), z, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                } else {
                    const float h = t.weights[slot] * (z > 0.0f ? z : 0.0f);
                    const uint16_t hi = act_cast<DT>(h, false);
                    const float back = to_float<DT>(hi);
                    const uint16_t lo = __builtin_fabsf(back) < __builtin_inff() ? act_cast<DT>(h - back, false) : (uint16_t)0;
                    uint16_t* const to = a.mid + (size_t)slot * (size_t)a.mid_row * 2 + (size_t)(n0 + c);
                    to[0] = hi;
                    to[a.mid_row] = lo;
                }
            }
        };
        const int pieces = WIDE || ODD ? scale_blocks : (a.in + 63) / 64, p0 = from(pieces, split), p1 = from(pieces, split + 1);
        floatx4 acc[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) acc[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (ODD) {
            expert_sums<DT, STORE, SECOND, NB, WAVES>(acc, rx, row_of_x(row0 + r16), (uint32_t)a.mid_row * 2u, w, scales, a.ld, n0, a.in, a.out,
                                                      p0, p1, wave, lane);
        } else {
            const uint32_t x_row[2] = {row_of_x(row0 + lane / 8), row_of_x(row0 + 8 + lane / 8)};
            const auto stream = [&](auto once) __attribute__((always_inline)) {
                expert_stream<DT, STORE, SECOND, once.value, NB, S, WAVES>(acc, a.x, x_bytes, x_row, (uint32_t)a.mid_row * 2u, w, scales, a.ld,
                                                                           n0, a.in, a.out, p0, p1, smem + wave * (S * STAGE),
                                                                           unit % max(p1 - p0, 1), wave, lane);
            };
            // (A branch for every piece costs 24 tokens 131 -> 140 us, both loops one token 24.3 -> 25.4.)
            if constexpr (KIND == 1) {
                if (a.once) stream(std::true_type{});
                else stream(std::false_type{});
            } else {
                stream(std::false_type{});
            }
        }
        finish(acc);
        if constexpr (SECOND) {
            wait_vmcnt<0>();           // this wave's sums have reached device scope
            __syncthreads();
            if (tid == 0) before = __hip_atomic_fetch_add(a.counters + nb, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            if (before == tiles * a.splits - 1) {
                asm volatile("" ::: "memory");   // the loads below stay after the count that allowed them
                // A token's parts are neighbours: (choice, part of k).  Several are loaded at once.
                const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.part, (uint32_t)(a.tokens * a.top * a.splits) * (uint32_t)a.out * 4u);
                const int parts = a.top * a.splits;
                constexpr int OUTS = 4;          // outputs a thread has on their way
                for (int o0 = tid; o0 < a.tokens * COLS; o0 += OUTS * THREADS) {
                    float z[OUTS];
#pragma unroll
                    for (int q = 0; q < OUTS; ++q) z[q] = row_without(min((o0 + q * THREADS) / COLS, a.tokens - 1));
                    for (int i0 = 0; i0 < parts; i0 += 4) {
                        float v[OUTS][4];
#pragma unroll
                        for (int q = 0; q < OUTS; ++q)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int o = o0 + q * THREADS, token = min(o / COLS, a.tokens - 1), c = n0 + o % COLS;
                                const bool live = o < a.tokens * COLS && i0 + i < parts && c < a.out &&
                                                  t.ids[token * a.top + min(i0 + i, parts - 1) / a.splits] >= 0;
                                const uint32_t at = ((uint32_t)(token * parts + i0 + i) * (uint32_t)a.out + (uint32_t)c) * 4u;
                                v[q][i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, live ? at : kOobOffset, 0, kDeviceScope));
                            }
#pragma unroll
                        for (int q = 0; q < OUTS; ++q)
#pragma unroll
                            for (int i = 0; i < 4; ++i) z[q] += v[q][i];
                    }
#pragma unroll
                    for (int q = 0; q < OUTS; ++q) {
                        const int o = o0 + q * THREADS, token = o / COLS, c = n0 + o % COLS;
                        if (o < a.tokens * COLS && c < a.out) a.y[(size_t)token * (size_t)a.out + (size_t)c] = act_cast<DT>(z[q], false);
                    }
                }
                if (tid == 0) __hip_atomic_store(a.counters + nb, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
        __syncthreads();
    }
}

}  // namespace gemm_relu_hip
