// w4_launch.h -- how the grouped products with 4-bit weights are cut into
// blocks.  Plain host arithmetic, no HIP.  The rules go by what uniform routing
// gives; other routings are as right, with more or fewer blocks than meant.
#pragma once

namespace moe_lora {

// Slots that a shard of E_l of the E experts gets of n, one at least.  (With all
// n counted, a shard of 16 of 128 experts and 2048 tokens top-8 took 104 us a
// layer instead of 79, one of 32 of 256 and 8192 tokens 264 instead of 186:
// hidden 2048, inter 768, without LoRA.)
inline int w4_local_slots(int n_slots, int E, int E_l)
{
    const long long n = (long long)n_slots * E_l / E;
    return n > 1 ? (int)n : 1;
}

// Rows per work-list tile (16: few-row kernel, 32 or 64: many-row kernel), from
// the rows an expert gets and the slots the shard gets.  Layer times in us with
// 16 / 32 / 64 rows a tile (hidden 2048, inter 768, groups of 128, no LoRA), on
// 128 experts top-8: 12 rows 93 / 99 / 109, 20 rows 117 / 102 / 112, 32 rows 139 /
// 137 / 120, 128 rows 350 / 308 / 266.  With fewer experts 32 rows a tile stay
// ahead until there are blocks enough for 64: 32 experts, 64 rows each, 83 / 75 /
// 83, 128 rows 124 / 108 / 99 (96 rows, the worst choice found, 103 / 93 / 86); a
// shard of 16 of 128 experts, 64 rows each, 73 / 60 / 66, 256 rows 178 / 120 /
// 111.  And 16 while a batch is a handful of tiles: 8 experts, 32 rows each, 40 /
// 45 / 51.
inline int w4_tile_rows(int n_slots, int E, int E_l)
{
    const int mean = n_slots / E, local = w4_local_slots(n_slots, E, E_l);
    if (mean <= 16 || local <= 320)
        return 16;
    return mean >= 24 && local >= 4096 ? 64 : 32;
}

// Few-row kernel: log2 of the shares of K per slab, for about `tiles` row tiles
// with rows.  1 share when the slabs alone make a wave per SIMD, doubling until
// they do or a share has no step left.
inline int w4_k_shares_log(int tiles, int n_slabs, int steps)
{
    const long long slabs = (long long)tiles * n_slabs;
    int log = 0;
    while (log < 3 && (slabs << log) < 1024 && (steps >> (log + 1)) >= 1)
        ++log;
    return log;
}

// Many-row kernel: row tiles with rows, of the n_tiles there may be, for a shard
// with n_local slots on n_busy experts.
inline int w4_row_tiles(int n_tiles, int n_busy, int n_local, int tile_rows)
{
    const int n = n_local / tile_rows > n_busy ? n_local / tile_rows : n_busy;
    return n < n_tiles ? n : n_tiles;
}

// Many-row kernel: slab groups (256 columns) that a block runs in turn on its
// row tile, for about `tiles` row tiles with rows and n_sg groups.  As few jobs
// per tile as still make kMinBlocks blocks, four rounds of two blocks per CU, and
// the groups spread evenly over them.  With 512 / 1024 / 2048 / 4096 blocks a
// layer of 128 experts top-8 (hidden 2048, inter 768, rank 64) takes 449 / 410 /
// 409 / 409 us at 2048 tokens and 898 / 732 / 703 / 712 at 4096.
constexpr int kMinBlocks = 2048;

inline int w4_groups_per_block(int tiles, int n_sg)
{
    int per = 1;
    while (per < n_sg && (long long)tiles * ((n_sg + per) / (per + 1)) >= kMinBlocks)
        ++per;
    const int jobs = (n_sg + per - 1) / per;
    return (n_sg + jobs - 1) / jobs;
}

} // namespace moe_lora
