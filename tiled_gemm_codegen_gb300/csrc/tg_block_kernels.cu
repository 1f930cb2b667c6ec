// One mode of block_kernel (-DTG_BLOCK_MODE=0 .. 3: BLOCK_GATED ..) in its tile
// shapes.
#include "tg_block.cuh"

#ifndef TG_BLOCK_MODE
#error "compile with -DTG_BLOCK_MODE"
#endif

namespace tg {
namespace {

template <int BN, int STAGES, bool PAIR>
BlockShape shape()
{
    constexpr int smem = Geometry<BN, PAIR>::smem_bytes(STAGES);
    static_assert(smem <= SMEM_LIMIT, "shared memory budget");
    return {block_kernel<TG_BLOCK_MODE, BN, STAGES, PAIR>, BN, smem, PAIR};
}

}  // namespace

#if TG_BLOCK_MODE == 0
BlockShape block_shape_gated(BlockTiles t)
#elif TG_BLOCK_MODE == 1
BlockShape block_shape_grad(BlockTiles t)
#elif TG_BLOCK_MODE == 2
BlockShape block_shape_shrink(BlockTiles t)
#else
BlockShape block_shape_adapt(BlockTiles t)
#endif
{
#if TG_BLOCK_MODE != 2  // (the adapters' first products have few features)
    if (t == TILES_PAIR) return shape<256, 6, true>();
#endif
    return t == TILES_FEW ? shape<32, 9, false>() : shape<128, 6, false>();
}

}  // namespace tg
