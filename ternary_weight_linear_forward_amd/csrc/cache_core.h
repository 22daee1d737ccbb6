// cache_core.h -- places of the int8 key / value cache (layout in bitlinear.h),
// shared by the kernels that write, read and attend to it.
#pragma once

#include "common.h"
#include "launch.h"

namespace bl {

constexpr int CACHE_BLOCK = 64; // tokens of one transposed block of V

// First row (token 0 of the page) of a page's head, in units of tokens.
__device__ __forceinline__ int64_t cache_row0(const CacheView &c, int64_t page, int head)
{
    return (page * c.heads + head) * c.page_tokens;
}

// Byte of token t (of 64) in a 64-byte row of a block of V.  A lane (row d =
// lane % 16, g = lane / 16) of a 16-row matrix-core operand takes the 16 bytes
// at 16 g: keys 4g + {0..3} of the block's four 16-key tiles, in tile order.
__device__ __forceinline__ int cache_v_byte(int t)
{
    return 16 * ((t % 16) / 4) + 8 * (t / 32) + 4 * ((t % 32) / 16) + t % 4;
}

} // namespace bl
