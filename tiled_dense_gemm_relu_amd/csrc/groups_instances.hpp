// The kernel instances of gemm_relu_groups.h, as tables of kernel addresses
// (groups_table.hpp); for each dtype one translation unit fills each.
#pragma once

#include "groups_dma.hpp"
#include "groups_kernels.hpp"
#include "groups_outer.hpp"
#include "groups_skinny.hpp"

namespace gemm_relu_hip {

// The LDS-DMA tile of a position of kGroupTile.
template <int T, bool A_KMAJOR, bool B_KMAJOR>
struct GroupTile;
template <bool AK, bool BK>
struct GroupTile<0, AK, BK> { using Cfg = GroupDmaConfig<256, 256, 2, 2, 4, AK, BK, 0>; };
template <bool AK, bool BK>
struct GroupTile<1, AK, BK> { using Cfg = GroupDmaConfig<128, 128, 4, 2, 2, AK, BK, 4>; };
template <bool AK, bool BK>
struct GroupTile<2, AK, BK> { using Cfg = GroupDmaConfig<64, 64, 4, 2, 2, AK, BK, 4>; };

template <int DT, int T, bool B_NK>
void fill_rows_dma(GroupKernels& t)
{
    using Cfg = typename GroupTile<T, false, !B_NK>::Cfg;
    static_assert(Cfg::BM == kGroupTile[T] && Cfg::BN == kGroupTile[T] && Cfg::THREADS == kGroupThreads[T],
                  "host tile table out of date");
    t.rows_dma[T][B_NK][0][0] = (const void*)&rows_dma<Cfg, DT, 0, kAdaptNone>;
    t.rows_dma[T][B_NK][1][0] = (const void*)&rows_dma<Cfg, DT, 1, kAdaptNone>;
    if constexpr (T == 0) {
        t.rows_dma[T][B_NK][0][1] = t.rows_dma[T][B_NK][1][1] = (const void*)&rows_dma<Cfg, DT, 1, kAdaptFirst>;
    } else {
        t.rows_dma[T][B_NK][2][0] = (const void*)&rows_dma<Cfg, DT, 2, kAdaptNone>;
        t.rows_dma[T][B_NK][0][1] = (const void*)&rows_dma<Cfg, DT, 0, kAdaptAfter>;
        t.rows_dma[T][B_NK][1][1] = (const void*)&rows_dma<Cfg, DT, 1, kAdaptAfter>;
        t.rows_dma[T][B_NK][2][1] = (const void*)&rows_dma<Cfg, DT, 2, kAdaptAfter>;
    }
}

template <int DT, int T>
void fill_group_tile(GroupKernels& t)
{
    fill_rows_dma<DT, T, false>(t);
    fill_rows_dma<DT, T, true>(t);
    t.weight_dma[T][0] = (const void*)&weight_dma<typename GroupTile<T, true, true>::Cfg, DT, 0>;
    if constexpr (T > 0) t.weight_dma[T][1] = (const void*)&weight_dma<typename GroupTile<T, true, true>::Cfg, DT, 2>;
}

// The register-staged tiles of a position of kStagedTile.  The large one keeps
// four steps of loads in flight, three where a mask or odd rows need more
// registers, the small one three.
template <int T, bool AK, bool BK, int MASKED, bool ODD>
using StagedTile = GroupDmaConfig<kStagedTile[T], kStagedTile[T], 2, 2, 2, AK, BK, 4, T == 0 && !ODD && MASKED == 0 ? 4 : 3, MASKED, ODD>;

template <int DT, int T, bool B_NK, bool ODD, bool MANY>
void fill_grad(StagedKernels& t)
{
    // dA = D @ B^T: for B stored (K, N) B_NK is true here, and dB = A^T @ D (q is D)
    t.grad[T][B_NK][0][MANY] =
        (const void*)&grad_staged<StagedTile<T, false, !B_NK, 0, ODD>, StagedTile<T, true, true, 0, ODD>, DT, MANY>;
    t.grad[T][B_NK][1][MANY] = (const void*)&grad_staged<StagedTile<T, false, !B_NK, 1, ODD>,
                                                         StagedTile<T, true, true, B_NK ? 2 : 1, ODD>, DT, MANY>;
}

template <int DT, int T, bool B_NK, bool ODD>
void fill_staged(StagedKernels& t)
{
    using Rows = StagedTile<T, false, !B_NK, 0, ODD>;
    static_assert(Rows::THREADS == kStagedThreads, "host tile table out of date");
    t.rows[T][B_NK][0][0] = (const void*)&rows_dma<Rows, DT, 1, kAdaptNone, false>;
    t.rows[T][B_NK][0][1] = (const void*)&rows_dma<Rows, DT, 1, kAdaptNone, true>;
    t.rows[T][B_NK][1][0] = t.rows[T][B_NK][1][1] = (const void*)&rows_dma<Rows, DT, 1, kAdaptAfter, false>;
    fill_grad<DT, T, B_NK, ODD, false>(t);
    fill_grad<DT, T, B_NK, ODD, true>(t);
}

template <int DT, bool ODD>
StagedKernels make_staged_table()
{
    StagedKernels t{};
    fill_staged<DT, 0, false, ODD>(t);
    fill_staged<DT, 0, true, ODD>(t);
    fill_staged<DT, 1, false, ODD>(t);
    fill_staged<DT, 1, true, ODD>(t);
    return t;
}

template <int DT, int S, bool B_NK>
void fill_skinny(GroupKernels& t)
{
    constexpr int MB = kSkinnyBlocks[S];
    t.rows_skinny[S][B_NK][0][0] = (const void*)&rows_skinny<DT, B_NK, MB, false, kSkinnyPlain>;
    t.rows_skinny[S][B_NK][0][1] = (const void*)&rows_skinny<DT, B_NK, MB, false, kSkinnyAdapters>;
    t.rows_skinny[S][B_NK][0][2] = (const void*)&rows_skinny<DT, B_NK, MB, false, kSkinnyMasked>;
    t.rows_skinny[S][B_NK][1][0] = (const void*)&rows_skinny<DT, B_NK, MB, true, kSkinnyPlain>;
    t.rows_skinny[S][B_NK][1][1] = (const void*)&rows_skinny<DT, B_NK, MB, true, kSkinnyAdapters>;
    t.rows_skinny[S][B_NK][1][2] = (const void*)&rows_skinny<DT, B_NK, MB, true, kSkinnyMasked>;
}

template <int DT>
GroupKernels make_group_table()
{
    GroupKernels t{};
    fill_skinny<DT, 0, false>(t);
    fill_skinny<DT, 0, true>(t);
    fill_skinny<DT, 1, false>(t);
    fill_skinny<DT, 1, true>(t);
    fill_skinny<DT, 2, false>(t);
    fill_skinny<DT, 2, true>(t);
    fill_group_tile<DT, 0>(t);
    fill_group_tile<DT, 1>(t);
    fill_group_tile<DT, 2>(t);
    t.weight_outer[0][0] = (const void*)&weight_outer<DT, 0, false>;
    t.weight_outer[0][1] = (const void*)&weight_outer<DT, 0, true>;
    t.weight_outer[1][0] = (const void*)&weight_outer<DT, 1, false>;
    t.weight_outer[1][1] = (const void*)&weight_outer<DT, 1, true>;
    t.weight_outer[2][0] = (const void*)&weight_outer<DT, 2, false>;
    t.weight_outer[2][1] = (const void*)&weight_outer<DT, 2, true>;
    t.mask = (const void*)&relu_mask<DT>;
    t.pad = (const void*)&pad_rows<DT>;
    t.shrink[0][0][0] = (const void*)&adapter_shrink<DT, false, 1, 1>;
    t.shrink[0][0][1] = (const void*)&adapter_shrink<DT, false, 1, 2>;
    t.shrink[0][1][0] = (const void*)&adapter_shrink<DT, false, 2, 1>;
    t.shrink[0][1][1] = (const void*)&adapter_shrink<DT, false, 2, 2>;
    t.shrink[1][0][0] = (const void*)&adapter_shrink<DT, true, 1, 1>;
    t.shrink[1][0][1] = (const void*)&adapter_shrink<DT, true, 1, 2>;
    t.shrink[1][1][0] = (const void*)&adapter_shrink<DT, true, 2, 1>;
    t.shrink[1][1][1] = (const void*)&adapter_shrink<DT, true, 2, 2>;
    return t;
}

}  // namespace gemm_relu_hip
