// w4_launch.h -- how the grouped products with 4-bit weights are cut into
// blocks.  Plain host arithmetic, no HIP.
#pragma once

namespace moe_lora {

// Many-row kernel: slab groups (256 columns) that a block runs in turn on its
// row tile, for about `tiles` row tiles with rows and n_sg groups.  As few jobs
// per tile as still make kMinBlocks blocks (two rounds of two blocks per CU; 700
// to 4096: the same times; 400: +38%), and the groups spread evenly over them.
constexpr int kMinBlocks = 1024;

inline int w4_groups_per_block(int tiles, int n_sg)
{
    int per = 1;
    while (per < n_sg && (long long)tiles * ((n_sg + per) / (per + 1)) >= kMinBlocks)
        ++per;
    const int jobs = (n_sg + per - 1) / per;
    return (n_sg + jobs - 1) / jobs;
}

} // namespace moe_lora
