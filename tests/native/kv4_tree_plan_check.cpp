// Every launch of svdq_kv4_tree_attention that its size checks let through must
// be one that the runtime takes (fewer than 2^24 blocks of 256 threads), with no
// more splits of the keys than the workspace of svdq_kv4_attention holds.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "kv4_plan.h"

int main()
{
    std::vector<int> sizes, bounds = {1, 2, 16, 17, 700, 4096, 1 << 20, INT32_MAX};
    for (int e = 0; e < 25; ++e)
        for (int d = -1; d <= 1; ++d)
            if ((1 << e) + d >= 1) sizes.push_back((1 << e) + d);
    uint64_t checked = 0, bad = 0;
    for (int heads : sizes)
        for (int group : {1, 3, 8, 64})
            for (int T : sizes)
                for (int B : sizes) {
                    if (heads > 65535 || (int64_t)T * heads * group * 64 >= (1 << 30)) continue;
                    if ((int64_t)B * heads >= (1 << 24)) continue;
                    for (int dim : {64, 128})
                        for (int max_q : {1, 5, 64, T, INT32_MAX})
                            for (int max_kv : bounds) {
                                const svdq::KvPlan c = svdq::kv4_plan(T, B, heads, group, max_q, max_kv, 256);
                                const svdq::KvPlan p = svdq::kv4_tree_plan(T, B, heads, group, dim, max_q, max_kv, 256);
                                const int64_t blocks = svdq::kv4_blocks(p, B, heads);
                                ++checked;
                                if (p.q_tiles >= 1 && p.splits >= 1 && p.splits <= c.splits && p.split_steps >= 1 &&
                                    blocks >= 1 && blocks * 256 < ((int64_t)1 << 32))
                                    continue;
                                if (bad++ == 0)
                                    std::printf("T %d B %d heads %d group %d dim %d max_q %d max_kv %d: %lld blocks\n", T, B,
                                                heads, group, dim, max_q, max_kv, (long long)blocks);
                            }
                }
    std::printf("checked %llu launches, bad %llu\n", (unsigned long long)checked, (unsigned long long)bad);
    return bad ? 1 : 0;
}
