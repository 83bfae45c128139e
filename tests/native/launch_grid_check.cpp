// launch_grid covers every number of blocks that svdq_residual_norm comes to
// (rows of 8 channels, four to a block, fewer than 2^30 values; and every count
// around powers of two) with launches that the runtime takes: fewer than 2^32
// threads of 256-thread blocks along x, at most 65535 blocks along y, row
// numbers within int32.
#include <cstdint>
#include <cstdio>

#include "launch_grid.h"

static uint64_t checked = 0, bad = 0;

static void check(int64_t blocks)
{
    const svdq::LaunchGrid g = svdq::launch_grid(blocks);
    ++checked;
    const int64_t all = (int64_t)g.x * g.y;
    if (g.x >= 1 && g.y >= 1 && g.y <= 65535 && (int64_t)g.x * 256 < ((int64_t)1 << 32) && all >= blocks &&
        all - blocks < g.x && 4 * all < ((int64_t)1 << 31) && (g.y == 1) == (blocks * 256 < ((int64_t)1 << 32)))
        return;
    if (bad++ == 0) std::printf("%lld blocks: %u x %u\n", (long long)blocks, g.x, g.y);
}

int main()
{
    for (int64_t M = 1; M * 8 < (1 << 30); M += M < 100000 ? 1 : 997) check((M + 3) / 4);
    check((((int64_t)1 << 27) - 1 + 3) / 4);
    for (int e = 0; e <= 25; ++e)
        for (int64_t d = -3; d <= 3; ++d)
            if (((int64_t)1 << e) + d >= 1) check(((int64_t)1 << e) + d);
    std::printf("checked %llu counts, bad %llu\n", (unsigned long long)checked, (unsigned long long)bad);
    return bad ? 1 : 0;
}
