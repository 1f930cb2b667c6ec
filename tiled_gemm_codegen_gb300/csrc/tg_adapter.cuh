// Device pieces of the adapters' layout (see tg_block.cuh) that its kernels
// share.
#pragma once

#include <cuda_bf16.h>

#include "tg_block.h"

namespace tg {

// A tile of ADAPT's rows: its adapters' first place and number, its first block.
struct AdapterTile {
    int32_t first, count, blk0;
};
__device__ __forceinline__ AdapterTile adapter_tile(const BlockParams &p, int32_t t)
{
    const int4 v = __ldcg(p.tab.tile + t);
    return {v.x, v.y, v.z};
}

// u = hi + lo: rounded to bf16, and what that leaves.  hi rounds down where
// rounding would make an infinity; an infinity or NaN is hi's alone.
__device__ __forceinline__ void split_parts(float x, __nv_bfloat16 &hi, __nv_bfloat16 &lo)
{
    constexpr float MOST = 3.402823466e38f;
    hi = __float2bfloat16_rn(x);
    lo = __ushort_as_bfloat16(0);
    if (fabsf(x) <= MOST) {
        if (fabsf(__bfloat162float(hi)) > MOST) hi = __ushort_as_bfloat16(static_cast<uint16_t>(__float_as_uint(x) >> 16));
        lo = __float2bfloat16_rn(__fsub_rn(x, __bfloat162float(hi)));
    }
}

// Where hi of value r of a row's u stands for adapter i of its tile (row `in`
// of the tile, whose blocks begin at blk0), in values; lo stands a block,
// bn * 64 values, behind it.  r a multiple of 8: 16 bytes.
__device__ __forceinline__ int64_t adapter_at(int32_t i, int32_t r, int32_t blk0, int32_t in, int32_t bn, int32_t Rp)
{
    const int32_t col = i * Rp + r;
    return (static_cast<int64_t>(blk0 + (col >> 6) * 2) * bn + in) * 64 + (col & 63);
}

// Zeros in row `in` of a tile's blocks (count adapters) but for adapter i's
// columns (-1: all of them).  A warp a row.
__device__ __forceinline__ void zero_columns(const BlockParams &p, int32_t in, int32_t blk0, int32_t count, int32_t i, int lane)
{
    const int32_t own = i < 0 ? -1 : i * (p.Rp / 8), end = own + p.Rp / 8;  // its 16 bytes of hi
    const int32_t all = adapter_blocks(count, p.Rp) * 4;
    for (int32_t k = lane; k < all; k += 32)
        if (own < 0 || k < own || k >= end) {
            uint16_t *at = p.wide + adapter_at(0, k * 8, blk0, in, p.wide_bn, 0);
            *reinterpret_cast<uint4 *>(at) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4 *>(at + static_cast<int64_t>(p.wide_bn) * 64) = make_uint4(0u, 0u, 0u, 0u);
        }
}

// The same for `rows` rows of a tile from `in` on, by `threads` threads of which this
// is `id`.
__device__ __forceinline__ void zero_rows(const BlockParams &p, const AdapterTile &ad, int32_t i, int32_t in, int32_t rows, int32_t id,
                                          int32_t threads)
{
    const int32_t own = i * (p.Rp / 8), end = own + p.Rp / 8, all = adapter_blocks(ad.count, p.Rp) * 4;
    if (all == end - own) return;
    for (int32_t k = id; k < rows * all; k += threads) {
        const int32_t row = k / all, u = k - row * all;
        if (u >= own && u < end) continue;
        uint16_t *at = p.wide + adapter_at(0, u * 8, ad.blk0, in + row, p.wide_bn, 0);
        *reinterpret_cast<uint4 *>(at) = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4 *>(at + static_cast<int64_t>(p.wide_bn) * 64) = make_uint4(0u, 0u, 0u, 0u);
    }
}

}  // namespace tg
