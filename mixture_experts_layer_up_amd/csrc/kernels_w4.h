// kernels_w4.h -- argument blocks and host launchers of the 4-bit expert
// weights: quantising, packing and the grouped products.  Internal to the
// library; the public interface is include/moe_lora.h, the packed layout is
// in w4_layout.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe_lora {

struct QuantizeW4Args {
    const uint16_t *src;   // bf16 [E_l, K, N]
    uint8_t *codes;        // [E_l, K / 2, N]: row 2i in the low nibble, row 2i + 1 in the high
    uint16_t *scales;      // bf16 [E_l, ceil(K / group), N]
    uint8_t *zeros;        // [E_l, ceil(K / group), N], or null (z = 8)
    int E_l, K, N, group;
};

struct PackW4Args {
    const uint8_t *codes;
    const uint16_t *scales;
    const uint8_t *zeros;  // or null
    uint8_t *dst;          // w4_layout(E_l, K, N, group, zeros).bytes
    int E_l, K, N, I;      // I > 0: gate/up interleaved tile order (w13)
    int group;
};

// Grouped expert product with 4-bit weights, the LoRA expand folded in.
struct GemmW4Args {
    const uint16_t *X;        // gate_up: hidden [T, K]; down: act [n, K]
    int K;
    const uint8_t *codes;     // the packed weight's regions (w4_layout.h)
    const uint16_t *scales;
    const uint8_t *zeros;     // or null
    int k_units, n_groups, group;
    int n_slabs;              // 64-column slabs per expert
    const uint16_t *S;        // shrink outputs [n, rp] by slot x, or null
    const uint16_t *LB;       // [L, E_l (shared: 1), n_canon, r] or null
    int r, rp, L, n_canon;    // n_canon: output columns of the unpacked weight
    int lb_shared, lb_stacks; // one LB stack per adapter; stacks in LB
    const int32_t *mapping;   // [T] or null
    const int4 *tiles;        // work list written by the permute kernel
    const int32_t *tile_count;
    int n_tiles, tile_rows;   // list length (upper bound), rows per tile
    int n_local, n_busy;      // slots of this shard on average, and experts they can touch
    const int32_t *perm2exp;  // [n]
    int E_l, k, I;
    void *Y;                  // gate_up: bf16 act [n, I]; down: [n, n_canon]
    int y_f32;                // down: Y is fp32, else bf16
};

struct FinalizeF32Args {
    const float *Y;           // [n, H]
    const int32_t *exp2perm;  // [T*k]
    const float *weights;     // [T, k]
    uint16_t *out;            // [T, H]
    int T, H, k;
    float scale;
};

hipError_t launch_gemm_w4(const GemmW4Args &a, bool gated, hipStream_t s);
hipError_t launch_gemm_w4_many(const GemmW4Args &a, bool gated, hipStream_t s);  // tiles of 32, 64 rows
hipError_t launch_finalize_f32(const FinalizeF32Args &a, hipStream_t s);
hipError_t launch_pack_w4(const PackW4Args &a, hipStream_t s);
hipError_t launch_quantize_w4(const QuantizeW4Args &a, hipStream_t s);

} // namespace moe_lora
