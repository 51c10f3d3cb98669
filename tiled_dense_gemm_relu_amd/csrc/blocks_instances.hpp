// The kernel instances of gemm_relu_blocks for one pair of formats.
#pragma once

#include "blocks_dma.hpp"

namespace gemm_relu_hip {

using Blocks256 = BlockConfig<256, 256, 2, 2, 4>;
using Blocks128 = BlockConfig<128, 128, 4, 2, 2>;
using Blocks64 = BlockConfig<64, 64, 4, 2, 2>;
static_assert(Blocks256::BM == kBlockTile[0] && Blocks128::BM == kBlockTile[1] && Blocks64::BM == kBlockTile[2], "tiles");
static_assert(Blocks256::THREADS == kBlockThreads[0] && Blocks128::THREADS == kBlockThreads[1] &&
                  Blocks64::THREADS == kBlockThreads[2], "threads");

template <int FA, int FB>
BlocksKernels make_blocks_table()
{
    return BlocksKernels{{{(const void*)blocks_dma<Blocks256, FA, FB, false>, (const void*)blocks_dma<Blocks256, FA, FB, true>},
                          {(const void*)blocks_dma<Blocks128, FA, FB, false>, (const void*)blocks_dma<Blocks128, FA, FB, true>},
                          {(const void*)blocks_dma<Blocks64, FA, FB, false>, (const void*)blocks_dma<Blocks64, FA, FB, true>}}};
}

}  // namespace gemm_relu_hip
