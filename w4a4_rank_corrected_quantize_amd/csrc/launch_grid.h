// launch_grid.h -- block counts that one launch takes.  Host arithmetic alone:
// it needs no HIP header.
#pragma once

#include <stdint.h>

namespace svdq {

constexpr int64_t kMaxBlocks = (1 << 24) - 1;     // of 256 threads along x: fewer than 2^32 threads

// At least `blocks` blocks of 256 threads, as y rows of x; y is 1 up to kMaxBlocks.
struct LaunchGrid {
    uint32_t x, y;
};

inline LaunchGrid launch_grid(int64_t blocks)
{
    constexpr int64_t kRow = 1 << 22;
    if (blocks <= kMaxBlocks) return {(uint32_t)blocks, 1};
    return {(uint32_t)kRow, (uint32_t)((blocks + kRow - 1) / kRow)};
}

}  // namespace svdq
