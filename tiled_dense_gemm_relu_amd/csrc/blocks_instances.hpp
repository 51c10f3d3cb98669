// The kernel instances of gemm_relu_blocks for one pair of formats.
#pragma once

#include "blocks_dma.hpp"
#include "blocks_stream.hpp"

namespace gemm_relu_hip {

using Blocks256 = BlockConfig<256, 256, 2, 2, 4, 0>;
using Blocks128 = BlockConfig<128, 128, 4, 2, 2, 4>;
using Blocks64 = BlockConfig<64, 64, 4, 2, 2, 4>;
static_assert(Blocks256::BM == kBlockTile[0] && Blocks128::BM == kBlockTile[1] && Blocks64::BM == kBlockTile[2], "tiles");
static_assert(Blocks256::THREADS == kBlockThreads[0] && Blocks128::THREADS == kBlockThreads[1] &&
                  Blocks64::THREADS == kBlockThreads[2], "threads");

template <int FA, int FB, int S>
constexpr void fill_stream(BlocksKernels& t)
{
    t.stream[S][0] = (const void*)blocks_stream<FA, FB, false, S>;
    t.stream[S][1] = (const void*)blocks_stream<FA, FB, true, S>;
    if constexpr (S + 1 < kNumStreams) fill_stream<FA, FB, S + 1>(t);
}

template <int FA, int FB>
BlocksKernels make_blocks_table()
{
    BlocksKernels t{{{(const void*)blocks_dma<Blocks256, FA, FB, false>, (const void*)blocks_dma<Blocks256, FA, FB, true>},
                          {(const void*)blocks_dma<Blocks128, FA, FB, false>, (const void*)blocks_dma<Blocks128, FA, FB, true>},
                          {(const void*)blocks_dma<Blocks64, FA, FB, false>, (const void*)blocks_dma<Blocks64, FA, FB, true>}}, {},
                    (const void*)blocks_pair<Blocks64, FA, FB>};
    fill_stream<FA, FB, 0>(t);
    return t;
}

}  // namespace gemm_relu_hip
