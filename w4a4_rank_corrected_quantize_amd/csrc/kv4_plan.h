// kv4_plan.h -- how svdq_kv4_attention divides its work over blocks.  Host
// arithmetic alone: it needs no HIP header.
#pragma once

#include "launch_grid.h"

namespace svdq {

constexpr int kKv4ManyTiles = 2;                  // 16-row tiles per wave of a block of many rows

// Form, tiles of rows and splits of the keys, from the sizes and the caller's
// bounds.
struct KvPlan {
    bool many;
    int q_tiles, splits, split_steps;             // a split's least length (many rows: its length within the bound)
};

inline KvPlan kv4_plan(int T, int B, int heads, int group, int max_q, int max_kv, int cus)
{
    KvPlan p;
    const int64_t rows = (int64_t)(max_q < T ? max_q : T) * group;
    p.many = rows > 16;
    const int block_rows = p.many ? 64 * kKv4ManyTiles : 16;
    const int64_t tiles = (rows + block_rows - 1) / block_rows;
    // blocks of rows: at most every sequence's, and the rows' own number and one more per sequence
    int64_t blocks = (int64_t)T * group / block_rows + B;
    blocks = (blocks < tiles * B ? blocks : tiles * B) * heads;
    // Splits.  Many rows: none where the rows alone give two blocks per compute
    // unit (a split writes and reads their fp32 sums), else about four blocks (8
    // sequences of 1 .. 700 rows over up to 6000 keys, 16 heads over 4: 2 blocks
    // 129 us, 3 124, 4 107, 6 107, 8 115), of at least four steps.
    // Few rows: none up to 12 steps (700 keys: 10.1 us, split 10.6); up to a block
    // per compute unit of at least four steps, one per wave (8000 keys, 8 heads:
    // 9.3 us, of eight 10.9); beyond that up to six of at least 16 (2 x 16000
    // keys: 17 us, of four steps 25).  Sequences shorter than the bound take as
    // many parts of that least length (one of 1500 keys under a bound of 32768:
    // 10.3 us, in parts of the bound's length 13.0).
    const int64_t steps = ((int64_t)max_kv + 63) / 64;
    auto up = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
    auto least = [](int64_t x, int64_t y) { return x < y ? x : y; };
    int64_t s, least_steps = 0;
    if (p.many) {
        s = blocks >= 2 * (int64_t)cus ? 1 : least(up(steps, 4), up(4 * (int64_t)cus, blocks));
    } else {
        const int64_t a = least(up(steps, 4), up(cus, blocks)), b = least(up(steps, 16), up(6 * (int64_t)cus, blocks));
        s = steps <= 12 ? 1 : (a > b ? a : b), least_steps = a >= b ? 4 : 16;
    }
    s = s > 64 ? 64 : s;
    p.split_steps = (int)((steps + s - 1) / s + 3) & ~3;
    p.splits = (int)((steps + p.split_steps - 1) / p.split_steps);
    if (!p.many) p.split_steps = (int)least_steps;
    // the runtime takes fewer than 2^32 threads along x; a block takes further tiles in a loop
    const int64_t cap = kMaxBlocks / ((int64_t)B * heads * p.splits);
    p.q_tiles = (int)(tiles > cap ? cap : tiles);
    return p;
}

// Blocks of 256 threads of the first kernel.
inline int64_t kv4_blocks(const KvPlan &p, int B, int heads) { return (int64_t)p.q_tiles * p.splits * B * heads; }

}  // namespace svdq
