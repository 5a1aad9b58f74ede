// cb3_blocks.h -- the 16-byte blocks of memory that hold a step of a 3-bit row (words of
// 10 codes): plain arithmetic, for the kernels and for a host program.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif

namespace moe {

struct Cb3Block {
    int at;          // first byte, counted from the row's start (may lie before it)
    uint32_t bytes;  // bytes up to the row's end, at most 16
};

// Block k (0 to 4) of the 128 codes from 128 j on, of a row of row_bytes bytes that starts
// `misplaced` words past a 16-byte boundary. A copy's source has to be aligned to its size
// even where none of it is read: past the row's end it is the block the row starts in.
MOE_HD Cb3Block cb3_block(uint32_t misplaced, uint32_t j, uint32_t k, uint32_t row_bytes) {
    const int word = (int)(128u * j / 10u), off = (int)((misplaced + (uint32_t)word) & 3u);
    const int at = (word - off) * 4 + (int)k * 16, n = (int)row_bytes - at;
    return {n > 0 ? at : -4 * (int)(misplaced & 3u), n >= 16 ? 16u : n > 0 ? (uint32_t)n : 0u};
}

}  // namespace moe
