// kernels_block.h -- argument blocks and host launchers of what stands around
// the layer in a block: products with an epilogue, block norms, clipping.
// Internal to the library; the public interface is include/moe_lora.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe_lora {

// ---- products -------------------------------------------------------------

// What happens to a sum before it is stored.  Columns of the product are those
// of the weight as the kernel reads it: `half` columns a projection (a multiple
// of 8 where a padded copy is read, else N), one projection or, for swiglu, two.
struct Epilogue {
    const float *bias;         // [W] or null
    const uint16_t *residual;  // [M, N] or null
    void *out;                 // [M, N]
    uint16_t *preact;          // [M, W] or null
    int N;                     // output columns
    int half;                  // columns of a projection in the weight as read
    int sets;                  // 1, or 2: the stored row has W = sets N columns
    int act;                   // MOE_LORA_ACT_*
    int fp32;                  // type of out
    int wide;                  // N and every pointer allow eight elements at once
    int padded;                // gradient of a padded weight: columns [N, half) are dropped
};

// out[m, n] = epilogue(sum_k Q[m, k] P[k, n]) over M rows, C columns of P and K
// terms.  Each operand is given with its contraction index contiguous (rows of
// length ld hold k) or strided (rows of length ld hold m or n); base pointers
// and ld * 2 bytes are multiples of 16.
struct ProductArgs {
    const uint16_t *Q, *P;
    int M, C, K;
    int ldq, ldp;
    int tiles_m, tiles_n;
    int splits, k_per;         // terms a split sums, a multiple of 64
    int64_t part;              // dz's second part (see ActGradArgs), in elements from the first; 0: none
    float *partial;            // [splits, M, C] when splits > 1
    Epilogue e;
};

enum class Product {
    forward,    // Q rows hold k, P rows hold n: x w
    input_grad, // Q rows hold k, P rows hold k: dz w^T
    weight_grad // Q rows hold m, P rows hold n: x^T dz
};

// Tile and split of a product; splits > 1 needs splits * M * C floats.
struct ProductPlan {
    int tile;      // index of the tile shape
    int tiles_m, tiles_n, splits, k_per;
    float us;      // estimate, without a launch's own time
};
// `parts` of a gradient: 2 double the steps.
ProductPlan plan_product(int64_t M, int64_t C, int64_t K, bool gated, int parts = 1);
hipError_t launch_product(Product kind, const ProductPlan &plan, const ProductArgs &a, hipStream_t s);
// The weight's and the input's gradient in one launch, with the same tiles, the input's
// whole: M rows, `in` and `columns` of the weight.  Returns the estimated microseconds.
float plan_both(int64_t M, int64_t in, int64_t columns, int parts, ProductPlan *dw, ProductPlan *dx);
hipError_t launch_both_gradients(const ProductPlan &dw, const ProductArgs &w, const ProductPlan &dx,
                                 const ProductArgs &x, hipStream_t s);

// The forward product for few rows or few outputs: the weight as given, any N.
struct RowsArgs {
    const uint16_t *x, *w;
    int M, K, W;
    Epilogue e;
};
struct RowsPlan {
    int mt, cpl;   // sixteens of rows a block takes, columns a lane loads; mt 0: too large
    float us;      // estimate
};
RowsPlan plan_rows(int64_t M, int64_t K, int64_t N, int sets);
hipError_t launch_rows(const RowsPlan &plan, const RowsArgs &a, hipStream_t s);

// Copy of w [K, sets N] with each projection padded by zeros to `half` columns.
hipError_t launch_pad_columns(const uint16_t *w, uint16_t *out, int64_t K, int N, int half, int sets,
                              hipStream_t s);

// dz = d_out act'(preact) as bf16 [M, sets half] (null: not wanted) and partial
// column sums [blocks, W] (null: not wanted), then d_bias [W] from them.  With `part`
// dz is the sum of two bf16 values, the second `part` elements behind the first.
struct ActGradArgs {
    const void *d_out;
    const uint16_t *preact;
    uint16_t *dz;
    float *partial;
    float *d_bias;
    int64_t M, part;
    int N, half, sets, act, fp32;
    int blocks;                // row strips
};
int act_grad_blocks(int64_t M);
hipError_t launch_act_grad(const ActGradArgs &a, hipStream_t s);

// out[q][c] = sum over r of in[r, q, c], q < sums <= 3, r in a fixed order: joins
// the column sums that blocks kept apart.
hipError_t launch_column_sums(const float *in, int rows, int sums, int columns, float *const *out,
                              hipStream_t s);

// ---- norms ----------------------------------------------------------------

struct NormArgs {
    const uint16_t *x, *y;     // residual, branch; [T, H] or null
    const uint16_t *w_post, *w_pre;
    const void *gate;
    uint16_t *r, *z;           // new residual, normed; or null
    int T, H, gate_kind;
    float eps, alpha, offset;
};
hipError_t launch_block_norm(const NormArgs &a, hipStream_t s);

struct NormGradArgs {
    const uint16_t *r, *y, *w_post, *w_pre;
    const void *gate;
    const uint16_t *dr, *dz;
    uint16_t *dx, *dy;
    float *d_token;            // gate gradient of tokens [T], or null
    float4 *stats;             // [T] for rows of more than 8192 columns
    float *partial;            // [blocks, sums, H]
    int post_at, pre_at, gate_at;  // place of each column sum, -1: not wanted
    int sums;
    int T, H, gate_kind, blocks;
    float eps, alpha, offset;
};
int norm_grad_blocks(int T, int H);
size_t norm_grad_stats_bytes(int T, int H);
hipError_t launch_block_norm_backward(const NormGradArgs &a, hipStream_t s);

// ---- clipping -------------------------------------------------------------

constexpr int kClipTensors = 112;     // tensors of one launch: the table is a kernel argument
constexpr int kClipLargest = 32768;   // elements of a block, at most

struct ClipTensor {
    const void *data;
    void *out;
    int64_t n;                 // elements
    int first;                 // first block of this tensor in its launch
    int fp32;
};

struct ClipTable {
    ClipTensor t[kClipTensors];
    int count;
    int blocks;
    int chunk;                 // elements of one block
    bool stream;               // results are written past the caches
};

// The factor of a call as power * rest; power is 1 where the product is a normal fp32
// value, else a power of two.  Both 1: leave the values as they are.
struct ClipFactor {
    float power, rest;
};

// What all blocks of a call share: partial[block] = sum of squares of the block's chunk,
// and what comes of their sum.
struct ClipSums {
    double *partial;
    int64_t blocks;            // of all launches
    float *norm;
    ClipFactor *factor;
    float max_norm;
};

hipError_t launch_clip_squares(const ClipTable &t, double *partial, hipStream_t s);
// Norm and factor from all partial sums, needed before the scaling of more than
// kClipFew blocks; fewer are summed by each scaling block, the first of which
// (`first_table`) writes the norm.
constexpr int64_t kClipFew = 4096;
hipError_t launch_clip_norm(const ClipSums &c, hipStream_t s);
hipError_t launch_clip_scale(const ClipTable &t, const ClipSums &c, bool first_table, hipStream_t s);

} // namespace moe_lora
