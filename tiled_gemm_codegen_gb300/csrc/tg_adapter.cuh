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

// Where a row's parts for adapter i of its tile begin (row `in` of the tile,
// whose blocks begin at blk0), in units of 8 values.
__device__ __forceinline__ int32_t adapter_unit(int32_t i, int32_t blk0, int32_t in, int32_t bn, int32_t Rp)
{
    const int32_t per = Rp <= 32 ? 32 / Rp : 1;
    const int32_t blk = blk0 + (Rp <= 32 ? i / per : i * (Rp / 32));
    return (blk * bn + in) * 8 + (Rp <= 32 ? i % per * (Rp / 4) : 0);
}

// Zeros in row `in` of a tile's blocks (count adapters) but for adapter i's
// columns (-1: all of them).  A warp a row.
__device__ __forceinline__ void zero_columns(const BlockParams &p, int32_t in, int32_t blk0, int32_t count, int32_t i, int lane)
{
    const int32_t units = p.Rp <= 32 ? p.Rp / 4 : p.Rp / 32 * 8;  // 16 bytes each, an adapter's
    const int32_t own = i * units, own_end = i < 0 ? own : own + units;
    for (int32_t k = lane; k < adapter_blocks(count, p.Rp) * 8; k += 32)
        if (k < own || k >= own_end)
            *reinterpret_cast<uint4 *>(p.wide + (static_cast<int64_t>(blk0 + (k >> 3)) * p.wide_bn + in) * 64 + (k & 7) * 8) =
                make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace tg
