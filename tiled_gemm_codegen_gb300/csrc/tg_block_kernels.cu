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
    using G = Geometry<BN, PAIR>;
    constexpr int bytes = STAGES * G::STAGE + block_epi_bytes(TG_BLOCK_MODE, BN) + block_bar_bytes(TG_BLOCK_MODE) + G::ALIGN_SLACK;
    constexpr int smem = bytes > G::ONE_CTA_PER_SM ? bytes : G::ONE_CTA_PER_SM;
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
    constexpr int STAGES = block_epi_bytes(TG_BLOCK_MODE, 256) > 32768 ? 5 : 6;
#if TG_BLOCK_MODE != 2  // (the adapters' first products have few features)
    if (t == TILES_PAIR) return shape<256, STAGES, true>();
#endif
    return t == TILES_FEW ? shape<32, 9, false>() : shape<128, STAGES, false>();
}

}  // namespace tg
