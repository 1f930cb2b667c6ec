// Agreement between the warps of a block.
#pragma once

#include <cstdint>

namespace tg {

// `threads` threads agree on a predicate (named barrier `id`, a multiple of 32
// of them): where waits may run out, the threads that meet at later barriers
// leave together or not at all.
__device__ __forceinline__ bool agree(bool pred, uint32_t id, uint32_t threads)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(pred)), "r"(id), "r"(threads)
        : "memory");
    return r != 0;
}

}  // namespace tg
