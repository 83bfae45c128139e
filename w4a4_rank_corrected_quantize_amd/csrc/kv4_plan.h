// kv4_plan.h -- how svdq_kv4_attention divides its work over blocks.  Host
// arithmetic alone: it needs no HIP header.
#pragma once

#include "launch_grid.h"

namespace svdq {

constexpr int kKv4ManyTiles = 2;                  // 16-row tiles per wave of a block of many rows

// Even division of the tree attention's work: parts of a tile's keys that the
// workspace holds, beyond the splits of the fixed division.
constexpr int kKv4EvenParts = 2;

// Form, tiles of rows and splits of the keys, from the sizes and the caller's
// bounds.
struct KvPlan {
    bool many;
    int q_tiles, splits, split_steps;             // a split's least length (many rows: its length within the bound)
};

inline KvPlan kv4_plan_form(bool many, int T, int B, int heads, int group, int max_q, int max_kv, int cus)
{
    KvPlan p;
    const int64_t rows = (int64_t)(max_q < T ? max_q : T) * group;
    p.many = many;
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

inline KvPlan kv4_plan(int T, int B, int heads, int group, int max_q, int max_kv, int cus)
{
    return kv4_plan_form((int64_t)(max_q < T ? max_q : T) * group > 16, T, B, heads, group, max_q, max_kv, cus);
}

// Trees of drafted tokens: more than 16 rows go 16 to a block as well while these
// are few.  A block of many rows takes as long per step for 17 rows as for 128 (heads
// of 128 1.3 us, one of 16 rows 0.3), so that 16 x 8 tokens over 8000 keys, 32 heads
// over 8 of 64, INT4, take 39 us instead of 67, 8 over 1000 keys 9 instead of 15;
// beyond a block per compute unit (heads of 64: three) it loses (16 x 16 tokens over
// 8000 keys, heads of 128, MXFP4: 106 and 91 us; of 64 58 and 70).  At most as many
// splits as kv4_plan has, so that its workspace serves both.
inline KvPlan kv4_tree_plan(int T, int B, int heads, int group, int dim, int max_q, int max_kv, int cus)
{
    const KvPlan p = kv4_plan(T, B, heads, group, max_q, max_kv, cus);
    if (!p.many) return p;
    const int64_t rows = (int64_t)(max_q < T ? max_q : T) * group, per = (rows + 15) / 16, own = (int64_t)T * group / 16 + B;
    if ((per * B < own ? per * B : own) * heads > (dim == 64 ? 3 : 1) * (int64_t)cus) return p;
    KvPlan f = kv4_plan_form(false, T, B, heads, group, max_q, max_kv, cus);
    if (f.splits > p.splits) f.splits = p.splits;
    return f;
}

// Blocks of 256 threads of the first kernel.
inline int64_t kv4_blocks(const KvPlan &p, int B, int heads) { return (int64_t)p.q_tiles * p.splits * B * heads; }

}  // namespace svdq
