// The kernel instances of gemm_relu_groups.h for one dtype, as a table of
// kernel addresses (groups_table.hpp); each dtype's translation unit fills one.
#pragma once

#include "groups_dma.hpp"
#include "groups_kernels.hpp"

namespace gemm_relu_hip {

template <int DT, int W>
void fill_group_width(GroupKernels& t)
{
    constexpr int VEC = kLoadWidths[W];
    t.rows_tiled[0][W] = (const void*)&rows_tiled<DT, false, VEC>;
    t.rows_tiled[1][W] = (const void*)&rows_tiled<DT, true, VEC>;
    t.weight_tiled[W] = (const void*)&weight_tiled<DT, VEC>;
}

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
    t.rows_dma[T][B_NK][0][0] = (const void*)&rows_dma<Cfg, DT, false, kAdaptNone>;
    t.rows_dma[T][B_NK][1][0] = (const void*)&rows_dma<Cfg, DT, true, kAdaptNone>;
    if constexpr (T == 0) {
        t.rows_dma[T][B_NK][0][1] = t.rows_dma[T][B_NK][1][1] = (const void*)&rows_dma<Cfg, DT, true, kAdaptFirst>;
    } else {
        t.rows_dma[T][B_NK][0][1] = (const void*)&rows_dma<Cfg, DT, false, kAdaptAfter>;
        t.rows_dma[T][B_NK][1][1] = (const void*)&rows_dma<Cfg, DT, true, kAdaptAfter>;
    }
}

template <int DT, int T>
void fill_group_tile(GroupKernels& t)
{
    fill_rows_dma<DT, T, false>(t);
    fill_rows_dma<DT, T, true>(t);
    t.weight_dma[T] = (const void*)&weight_dma<typename GroupTile<T, true, true>::Cfg, DT>;
}

template <int DT>
GroupKernels make_group_table()
{
    GroupKernels t{};
    fill_group_width<DT, 0>(t);
    fill_group_width<DT, 1>(t);
    fill_group_width<DT, 2>(t);
    fill_group_width<DT, 3>(t);
    fill_group_tile<DT, 0>(t);
    fill_group_tile<DT, 1>(t);
    fill_group_tile<DT, 2>(t);
    t.mask = (const void*)&relu_mask<DT>;
    t.shrink[0] = (const void*)&adapter_shrink<DT, false>;
    t.shrink[1] = (const void*)&adapter_shrink<DT, true>;
    return t;
}

}  // namespace gemm_relu_hip
